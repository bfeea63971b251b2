"""The delta on a stream that is given, with workspaces that the calls allocate."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("T,mode", [(16, "auto"), (16, "bgmv"), (700, "sgmv")])
def test_workspaces_of_another_stream(raw, T, mode):
    """They are neither still in use on the current stream, nor reused there or cleared
    too late."""
    import segmented_gather_rank_amd as L

    g = torch.Generator("cuda").manual_seed(T)
    r = lambda *s: (0.1 * torch.randn(s, generator=g, device="cuda")).bfloat16()  # noqa: E731
    x, A, B = r(T, 512), r(4, 512, 16), r(4, 16, 768)
    slots = torch.randint(-1, 4, (T,), generator=g, device="cuda", dtype=torch.int32)

    def call(stream):
        meta = L.lora_prepare_meta(slots, 4, stream=stream)
        L.lora_apply(meta, x, [A], [B], [0], y, add=False, mode=mode, stream=stream)
        return meta

    y = torch.zeros((T, 768), dtype=torch.bfloat16, device="cuda")
    call(None)
    torch.cuda.synchronize()
    want = y.clone()
    sizes = [L.lora_meta_workspace_bytes(T, 4),
             max(L.APPLY_SYNC_BYTES, L.lora_apply_workspace_bytes(T, 4, 512, 1, 16, torch.bfloat16, mode))]
    busy = torch.randn((4096, 4096), device="cuda")
    s = torch.cuda.Stream()
    for size in sizes:
        y.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            busy.mul_(1.0001)
        held = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        del held
        meta = call(s.cuda_stream if raw else s)
        for _ in range(4):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del meta
        assert torch.equal(y, want)
