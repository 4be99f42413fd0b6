"""CPU checks of the training operators' C ABI: exports and the argument checks
that answer without a GPU."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "domino_train.h")


def _declared():
    return sorted(set(re.findall(r"DOMINO_API\s+[\w\s\*]+?\b(domino_\w+)\s*\(", open(HEADER).read())))


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_lm_gb300 import build, rollout, train
    if not os.path.exists(rollout.LIB_PATH):
        build.build()
    return train.load_library()


def test_library_exports_every_declared_symbol(lib):
    from speculative_decoding_draft_lm_gb300 import train
    assert _declared() == sorted(train.EXPORTED)
    for name in _declared():
        assert hasattr(lib, name), name


def test_header_constants_match_the_binding():
    from speculative_decoding_draft_lm_gb300 import train
    text = open(HEADER).read()
    for name in ("DOMINO_TRAIN_MAX_V", "DOMINO_TRAIN_MAX_K", "DOMINO_TRAIN_MAX_TOKENS", "DOMINO_TRAIN_STATS"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(train, name)


def test_null_context(lib):
    from speculative_decoding_draft_lm_gb300 import rollout as R
    bad = R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_train_top_logits(None, None, 1, 8, 1, 1, 1.0, None, None, None, None) == bad
    assert lib.domino_train_distill_forward(None, None, 8, 1, None, None, None, 1, 1.0, None, None, None) == bad
    assert lib.domino_train_distill_backward(None, None, 8, 1, None, None, None, 1, 1.0, None, None, None, 8, None) == bad
    assert lib.domino_train_distill_step(None, None, 8, 1, None, None, None, 1, 1.0, None, None, None, 8, None) == bad
    assert lib.domino_train_embed(None, None, None, 1, 1.0, None, 8, None) == bad
    assert lib.domino_train_embed_grad(None, None, 8, None, 1, 1.0, None, 0, 0, None) == bad
    assert lib.domino_train_status(None, None) == bad
    assert lib.domino_train_last_launch_count(None) == 0
    lib.domino_train_destroy(None)


def test_config_validation_precedes_device_access(lib):
    from speculative_decoding_draft_lm_gb300 import rollout as R
    from speculative_decoding_draft_lm_gb300.train import domino_train_config as cfg
    ctx = ctypes.c_void_p()

    def init(*a):
        return lib.domino_train_init(ctypes.byref(ctx), ctypes.byref(cfg(*a)), 0)

    assert lib.domino_train_init(None, ctypes.byref(cfg(100, 8, 8, 1)), 0) == R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_train_init(ctypes.byref(ctx), None, 0) == R.DOMINO_ERR_INVALID_ARG
    assert init(100, 8, 8, 7) == R.DOMINO_ERR_UNSUPPORTED
    assert init(524289, 8, 8, 1) == R.DOMINO_ERR_UNSUPPORTED
    for bad in ((1, 8, 8, 1), (100, -1, 8, 1), (100, 8, -1, 1), (100, 8, 4194305, 1), (-5, 8, 8, 0)):
        assert init(*bad) == R.DOMINO_ERR_INVALID_ARG
    assert not ctx.value
