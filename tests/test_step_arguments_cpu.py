"""Refusals of the autograd forms that need no GPU."""
import pytest


@pytest.mark.parametrize("dtype", ["float16", "float64", "int32"])
def test_embedding_refuses_an_output_type(dtype):
    torch = pytest.importorskip("torch")
    from mxfp4_precision_gemms_gb300.step import embedding

    with pytest.raises(ValueError, match="out_dtype"):
        embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8), out_dtype=getattr(torch, dtype))
