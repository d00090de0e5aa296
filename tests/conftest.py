import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built libasyncpipe")
    # Tests without a GPU pass made-up device addresses, each in a call that its
    # checks refuse. Should a check be lost, such a call must find no device to
    # launch on: hidden here, before anything asks for one.
    if config.option.markexpr.replace(" ", "") == "notgpu":
        os.environ["CUDA_VISIBLE_DEVICES"] = ""


def pytest_collection_modifyitems(config, items):
    """In a session that has a device, the tests that rely on having none are skipped."""
    made_up = [i for i in items if i.path.name in ("test_fp8_cpu.py", "test_fp8_plans_cpu.py")]
    if not made_up:
        return
    try:
        import torch
    except ImportError:
        return
    if torch.cuda.is_available():
        for item in made_up:
            item.add_marker(pytest.mark.skip(reason="made-up device addresses, and a device is visible"))


@pytest.fixture(scope="session")
def orc():
    import oracle

    return oracle.load()
