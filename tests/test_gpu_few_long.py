"""Decode of few long (sequence, kv head) pairs: CTAs of eight (16-bit pools) and twelve warps
(8-bit pools) that take an SM each, in clusters of up to sixteen.  These run where a call has at most
an eighth as many pairs as SMs and a pair may show 256 blocks or more."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_b8 import run_attention  # noqa: E402
from test_gpu_window import run_decode  # noqa: E402

pytestmark = pytest.mark.gpu
MAXB = 420                                   # blocks: 6,720 tokens


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (12, 1), (32, 2)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("window,sinks", [(4500, 40), (2 ** 31 - 1, 0)])
def test_16bit(dtype, dim, hq, hkv, window, sinks):
    run_decode([6001, 0, 17, 4700], hq, hkv, dim, dtype, window, sinks, hq + dim, maxb=MAXB)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (12, 1), (32, 2)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("window,sinks", [(4500, 40), (None, 0)])
def test_8bit(dtype, dim, hq, hkv, window, sinks):
    run_attention([6001, 0, 17, 4700], hq, hkv, dim, dtype, window, sinks, hq + dim, maxb=MAXB)


@pytest.mark.parametrize("seqs", [1, 2, 5, 9, 19])
def test_cluster_sizes(seqs):
    """From sixteen CTAs a pair to the most pairs that this path takes."""
    lens = [6700 - 331 * i for i in range(seqs)]
    run_decode(lens, 2, 1, 64, "bf16", 2 ** 31 - 1, 0, seqs, maxb=MAXB)
    run_attention(lens, 2, 1, 64, "f16", None, 0, seqs, maxb=MAXB)
