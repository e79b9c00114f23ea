"""The dense calls with a stream of their own: outputs and workspaces that they allocate are not
memory that the current stream still uses, or gets before their kernels are done."""
import pytest
import torch

import tensorized_online_softmax_gb300 as fat

pytestmark = pytest.mark.gpu

B, H, N, D = 1, 4, 640, 128
WAIT = 40_000_000  # cycles: some 20 ms


def calls():
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn((B, H, N, D), generator=g).to(torch.bfloat16).cuda()
                   for _ in range(4))
    o, lse = fat.attn_fwd(q, k, v, True)
    host = [t.cpu().pin_memory() for t in (q, k, v)]
    return {
        "fwd": lambda s: fat.attn_fwd(q, k, v, True, stream=s),
        "splitkv": lambda s: fat.attn_fwd_splitkv(q, k, v, True, num_splits=3, stream=s),
        # (dQ: sums in no fixed order)
        "bwd": lambda s: fat.attn_bwd(q, k, v, o, lse, do, True, stream=s)[1:],
        "host": lambda s: fat.attn_fwd_host(*host, True, stream=s),
    }


def overwrite(times):
    """New tensors of every size that the calls allocate, filled, and let go of."""
    lib = fat.load_library()
    sizes = [4 * B * H * N * D] * 3 + [4 * B * H * N,
             lib.fat_attn_splitkv_workspace_bytes(B, H, N, D, 3),
             lib.fat_attn_bwd_workspace_bytes(B, H, N),
             lib.fat_attn_fwd_host_workspace_bytes(B, H, N, D, 0)]
    for t in [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes * times]:
        t.fill_(0xFF)


@pytest.mark.parametrize("name", ["fwd", "splitkv", "bwd", "host"])
def test_memory_of_a_call_on_another_stream(cuda_device, name):
    call = calls()[name]
    side = torch.cuda.Stream()
    out = call(None)
    torch.cuda.synchronize()  # (the host call's results are there once the stream is done)
    want = [t.clone() for t in out]
    for _ in range(2):
        call(side)
        overwrite(2)
    torch.cuda.synchronize()
    # the current stream still writes what it last let go of
    torch.cuda._sleep(WAIT)
    overwrite(1)
    got = call(side)
    side.synchronize()
    early = torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert not early, "the current stream was done too soon to show anything"
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the call's workspace is let go of on return, its kernels still to run
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    got = call(side)
    overwrite(2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert fat.check_device_error() == fat.FAT_OK


class Wrapped:
    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("name", ["fwd", "splitkv", "bwd", "host"])
def test_streams_given_in_other_ways(cuda_device, name):
    """A handle, an object that has one, the default stream by its numbers, and the per-thread
    default stream."""
    call = calls()[name]
    out = call(None)
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    side = torch.cuda.Stream()
    for stream in (side.cuda_stream, Wrapped(side), 0, 1, 2, torch.cuda.ExternalStream(side.cuda_stream)):
        got = call(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
