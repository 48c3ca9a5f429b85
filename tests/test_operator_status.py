"""Status words in the C ABI, without a GPU: bad arguments are refused before any device work."""
import ctypes

from test_operator_refusals import L, P, _append, _cache, _cfg, _w4  # noqa: F401


def test_a_status_word_needs_somewhere_to_go(L):  # noqa: F811
    assert L.lib.gmla_status_word(None) == L.GMLA_ERR_INVALID_ARG
    assert b"word" in L.lib.gmla_last_error()


def test_a_misaligned_status_is_refused(L):  # noqa: F811
    for status in (P + 1, P + 2):
        assert _append(L, cfg=_cfg(L, status=status)) == L.GMLA_ERR_INVALID_ARG
        assert b"status" in L.lib.gmla_last_error()
        assert _w4(L, cfg=_cfg(L, cache_dtype=0, status=status)) == L.GMLA_ERR_INVALID_ARG
        assert L.gmla_decode_workspace_size(_cfg(L, status=status), 4) == 256


def test_a_status_word_does_not_replace_the_workspace(L):  # noqa: F811
    assert _append(L, cfg=_cfg(L, status=P + 4), ws=None) == L.GMLA_ERR_WORKSPACE
    assert _append(L, cfg=_cfg(L, status=P + 4), cache=_cache(L, scales=None)) == L.GMLA_ERR_INVALID_ARG


def test_the_config_ends_with_the_status(L):  # noqa: F811
    assert L.gmla_config._fields_[-1] == ("status", ctypes.c_void_p) and L.gmla_config().status is None
