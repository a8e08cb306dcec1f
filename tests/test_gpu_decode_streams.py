"""The decode operators on a stream that is not the current one."""

import pytest
import torch

import orpo_preference_loss_gb300 as orpo
from gpu_helpers import dev, status_tensor

pytestmark = pytest.mark.gpu

M, D, V, GROUP = 512, 4096, 1000, 64


@pytest.fixture(scope="module")
def head():
    g = torch.Generator("cuda").manual_seed(1)
    wq = torch.randint(0, 256, (V, D // 2), generator=g, device=dev(), dtype=torch.uint8)
    sc = (torch.rand((V, D // GROUP), generator=g, device=dev()) * 0.01).bfloat16()
    return torch.randn((M, D), generator=g, device=dev()).bfloat16(), (wq, sc, (sc.float() * -7.5).bfloat16())


def test_own_workspace_on_a_side_stream_leaves_freed_blocks_alone(head):
    """A block that the current stream still has to read, freed on the host already, is not the workspace of a call
    on another stream; and what the current stream writes next does not reach that call's workspace."""
    h, q = head
    need = orpo.orpo_head_logits_q_workspace_bytes(M, D, 4)
    assert need > 1 << 20
    want = torch.empty((M, V), device=dev())
    st = status_tensor()
    orpo.orpo_head_logits_q(h, *q, 4, GROUP, 0.0, want, st)
    side = torch.cuda.Stream()
    for _ in range(3):
        out = torch.full((M, V), float("nan"), device=dev())
        block = torch.full((need,), 0x5A, dtype=torch.uint8, device=dev())
        copy = torch.empty_like(block)
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)  # a few hundredths of a second
        copy.copy_(block)
        del block
        orpo.orpo_head_logits_q(h, *q, 4, GROUP, 0.0, out, st, stream=side)
        again = torch.full((need,), 0xA5, dtype=torch.uint8, device=dev())
        torch.cuda.synchronize()
        assert torch.all(copy == 0x5A) and torch.all(again == 0xA5)
        assert torch.equal(out, want) and int(st.item()) == 0


def test_workspace_of_the_caller_on_a_side_stream(head):
    """Everything the call reads and writes is ready before the side stream starts, and kept until it ends."""
    h, q = head
    need = orpo.orpo_head_logits_q_workspace_bytes(M, D, 4)
    want, out = torch.empty((M, V), device=dev()), torch.full((M, V), float("nan"), device=dev())
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=dev())
    st = status_tensor()
    orpo.orpo_head_logits_q(h, *q, 4, GROUP, 0.0, want, st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    orpo.orpo_head_logits_q(h, *q, 4, GROUP, 0.0, out, st, stream=side, workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.all(ws[need:] == 0xFF) and int(st.item()) == 0
