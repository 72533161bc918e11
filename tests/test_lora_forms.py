"""Which form a forward pass of adapters takes, as the work memory that it asks for says (0: row by row).  The table of
adapters may be far larger than what a call uses, so that its size alone does not send a prompt to the form for
decoding rows."""
import pytest

from quantized_ffn_gb300 import build as zbuild
from quantized_ffn_gb300 import zffn


@pytest.fixture(scope="module")
def work():
    zbuild.build()
    return lambda T, r, L: zffn.load().zffn_lora_work_bytes(T, r, L, 0)


@pytest.mark.parametrize("T,r,L", [(1, 128, 1), (1, 8, 4096), (8, 16, 4), (61, 16, 48), (64, 64, 64), (512, 16, 64), (256, 16, 256), (1024, 16, 1024), (9, 40, 64), (40, 56, 64)])
def test_decoding_rows(work, T, r, L):
    assert work(T, r, L) == 0


@pytest.mark.parametrize("T,r,L", [(2048, 32, 256), (16384, 64, 4096), (1024, 16, 64), (512, 32, 128), (2048, 64, 512), (300, 40, 96), (64, 128, 1), (2048, 64, 8)])
def test_prompts(work, T, r, L):
    assert work(T, r, L) > 0


@pytest.mark.parametrize("r", [8, 24, 64, 128])
@pytest.mark.parametrize("L", [1, 8, 128, 4096])
def test_one_border(work, r, L):
    # from some number of tokens on it is always tiles
    forms = [work(T, r, L) > 0 for T in range(1, 20000, 37)] + [work(1 << 20, r, L) > 0]
    assert forms == sorted(forms) and forms[-1]
