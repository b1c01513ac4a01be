"""CPU: what the library's checks say to lists of no tokens, whose arrays have no address."""
import pytest

from sparse_attention_mla_gb300 import build_ext
import sparse_attention_mla_gb300 as dsa

from test_paged_host import FAKE, mla


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return dsa.load_library()


@pytest.mark.parametrize("call", [dict(B=0), dict(B=4, cu=FAKE)])
def test_lists_of_no_tokens_are_no_invalid_argument(lib, call):
    # (the status after the checks is that of the device, of which there may be none)
    assert mla(lib, N=0, K=7, q=None, out=None, lse=None, **call) != 3
    assert mla(lib, N=0, K=7, q=None, out=None, lse=None, wsb=0, **call) == 4


@pytest.mark.parametrize("bad", [dict(K=7), dict(idx=FAKE, K=0), dict(N=0, B=0, idx=FAKE, K=0)])
def test_lists_of_tokens_are_still_checked(lib, bad):
    assert mla(lib, **bad) == 3
