"""The timeout path of the prompt attention, by the library's own hook (rkv_debug_wait_fault): every CTA leaves
one load of K or V out, and every wait of the kernel gives up after 2e6 cycles, about a millisecond.  The kernel
has to report RKV_ERR_DEVICE_TIMEOUT, let its copies and products finish, free its tensor memory and return, and
the next calls on the same context have to give the bits of the calls before."""
import pytest
import torch

from _gpu_common import GUARD, assert_guards, ensure_lib, out_buffer
from reference_residual_kv_gb300 import rkv
from test_gpu_prompt import MARK, cache_with, i32, packed, randn, rows_kv

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
CYCLES = 2_000_000


def runs_out_and_goes_on(obj, call, shape, skip, written):
    """call(out) with `written` rows; obj holds the status."""
    def run():
        obj.status.zero_()
        out = out_buffer(shape, BF16)
        out.fill_(MARK)
        call(out)
        assert_guards(obj)
        assert bool((out.view(-1, *shape[-2:])[~written] == MARK).all())
        return out

    want = run()
    assert obj.device_status() == 0
    rkv.rkv_debug_wait_fault(CYCLES, skip)
    run()
    assert obj.device_status() == rkv.RKV_ERR_DEVICE_TIMEOUT
    for _ in range(2):                                       # the hook was one-shot
        again = run()
        assert obj.device_status() == 0 and torch.equal(again, want)


# items worked out by the producers, items split over the keys, items of the plan
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,H,N", [([700, 400], 8, 2), ([3000], 2, 1), ([300] * 40, 4, 2)])
@pytest.mark.parametrize("skip", [0, 1, 3])
def test_prompts(D, lens, H, N, skip):
    ensure_lib()
    gen = torch.Generator(device="cuda").manual_seed(D + skip)
    q, k, v, start = packed(gen, lens, H, N, D, behind=5)
    written = torch.arange(q.shape[0], device="cuda") < start[-1]
    h, st = rkv.PromptHeads(H, N, D, guard=GUARD), i32(start)
    runs_out_and_goes_on(h, lambda out: h.attend(q, k, v, st, out), q.shape, skip, written)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("skip", [0, 1, 2])
def test_pieces(D, skip):
    gen = torch.Generator(device="cuda").manual_seed(D + skip)
    S, n, T, H, N = 2, 150, 1500, 4, 2
    lens, new = [1300, 200], [150, 90]
    c = cache_with(rows_kv(gen, S, 1300, N, D), lens, T, N, D, 4)
    q, kv = randn(gen, S, n, H, D).to(BF16), rows_kv(gen, S, n, N, D)
    written = (torch.arange(n, device="cuda")[None] < i32(new)[:, None]).view(-1)
    ln, nn = i32(lens), i32(new)
    runs_out_and_goes_on(c, lambda out: c.chunk_attend(H, q, kv, ln, out, n_new=nn), q.shape, skip, written)
