"""A call that fails inside CUDA leaves no error behind: the check after the next
call's launch would report it as that one's. (A failure cannot be caused here
without a device, nor on one without disturbing it, so the source is read.)"""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_inner_product_b200", "csrc")


def _source(name):
    return open(os.path.join(CSRC, name)).read()


def test_every_failure_clears_the_error():
    """Both files of entry points report failures through cuda_fail, and that clears."""
    api = _source("tt_api.cu")
    body = api[api.index("tt_status cuda_fail("):]
    assert "cudaGetLastError();" in body[:body.index("\n}")]
    for name in ("tt_api.cu", "tt_train_api.cu"):
        text = _source(name)
        macro = text[text.index("#define TT_CUDA("):]
        assert "cuda_fail(" in macro[:macro.index("\n\n")], name
