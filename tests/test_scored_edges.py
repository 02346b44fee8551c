"""Arguments of the operators of changed scores and drafted trees that are refused although a kernel could be asked to run,
without a GPU."""
import pytest
import torch

from fp8_attention_forward_gb300 import build, fa8


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    fa8.lib()


@pytest.fixture(params=["c", "python"], autouse=True)
def entries(request, monkeypatch):
    """The views packed by the CPython module, and by the binding itself."""
    monkeypatch.setattr(fa8, "_entries", {})
    if request.param == "python":
        monkeypatch.setattr(fa8, "_args_module", lambda: None)
    elif fa8._args_module() is None:
        pytest.skip("Python's headers are missing here")


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("given", [dict(max_tokens=0), dict(masks=i32(7, 0))])
def test_packed_tokens_with_masks_of_no_words_are_refused(given):
    """Neither masks nor positions could be told from what lay there before."""
    with pytest.raises(fa8.Fa8Error) as e:
        fa8.tree_masks(i32(7), cu_seqlens_q=i32(3), **given)
    assert e.value.status == fa8.FA8_ERR_INVALID_ARG
    fa8.tree_masks(i32(0), cu_seqlens_q=i32(3), max_tokens=0)  # no tokens, nothing to do
