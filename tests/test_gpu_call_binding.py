"""The compiled marshalling of the prompt-side and shared-prefix calls (_calls)."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def plans(lib, cuda):
    q = torch.zeros((4, 2, 128), dtype=torch.bfloat16, device=cuda)
    K = torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16, device=cuda)

    def up(plan):
        return lib.TilePlan(plan, torch.from_numpy(plan).to(cuda))

    return q, K, up(lib.tg_plan_prefill([4], [4], 1, 2, 128, 1)[0]), up(lib.tg_plan_prefix([0, 4], [0], [[16]], 2, 1, 16, 128, 1)[0])


def test_the_interpreter_lock_is_given_up_for_the_call(lib, cuda, plans, monkeypatch):
    """In the place of the library's functions, one that tells whether its thread holds the lock."""
    q, K, prefill, prefix = plans
    _, _, calls = lib._setup()
    holds = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    real = [ctypes.cast(getattr(lib.load(), n), ctypes.c_void_p).value
            for n in ("tg_qk_norm_rope", "tg_prefill_attn", "tg_prefix_attn")]
    seen = []
    monkeypatch.setattr(lib, "_check", seen.append)  # called with anything but 0
    qkv = torch.zeros((4, 4, 128), dtype=torch.bfloat16, device=cuda)
    cu, start = torch.tensor([0, 4], dtype=torch.int32, device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
    pool = torch.zeros((1, 1, 2, 16, 128), dtype=torch.bfloat16, device=cuda)
    off, ids = torch.tensor([0, 1], device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
    try:
        calls.bind(holds, holds, holds)
        lib.tg_qk_norm_rope(qkv, cu, start, None, q, K, K.clone())
        lib.tg_prefill_attn(prefill, q, K, K.clone(), 1.0, q.clone())
        lib.tg_prefix_attn(prefix, q, pool, 1, off, ids, 1.0, q.clone())
    finally:
        calls.bind(*real)
    assert seen == []
