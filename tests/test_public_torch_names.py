"""The package uses torch through its public names: others may go with any release."""
import os
import re

import fp8_moe_expert_gb300 as fme


def test_no_private_torch_names():
    here = os.path.dirname(os.path.abspath(fme.__file__))
    for name in sorted(os.listdir(here)):
        if name.endswith(".py"):
            assert not re.findall(r"torch(?:\.\w+)*\._(?!_)\w+", open(os.path.join(here, name)).read()), name
