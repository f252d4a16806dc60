"""GPU test of what a handle of the gated linear recurrence allocates, against what the header states."""
import gc

import pytest
import torch

import random_feature_gb300 as R

pytestmark = pytest.mark.gpu

MB = 1 << 20


def stated(D, dtype, max_B, max_L, training):
    """Bytes, by the rule at favor_recur_create."""
    rows = max_B * -(-D // 128)
    places = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    blocks = max(rows, min(places, rows * min(64, -(-max_L // 64))))
    scan = 0 if max_L <= 8 else 9216 * blocks + 512 * rows
    return max(scan, 19968 * blocks + 1024 * rows * -(-max_L // (4 if dtype == "bf16" else 2))) if training else scan


# decoding handles, and ones for training from single tokens to long rows
@pytest.mark.parametrize("D,dtype,max_B,max_L,training", [
    (2048, "bf16", 256, 1, False), (2048, "f32", 512, 8, False), (2048, "bf16", 256, 1, True),
    (2048, "f32", 256, 1, True), (1536, "bf16", 8, 4096, False), (1, "f32", 1, 1 << 18, True),
    (64, "bf16", 8, 65536, True),
])
def test_workspace(D, dtype, max_B, max_L, training):
    """Free memory moves in blocks of 2 MB; what a process allocates in its first calls comes before."""
    with R.Recurrence(D, dtype, 1, 9) as f:
        f.new_state(1)
    gc.collect()        # handles of other tests
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    with R.Recurrence(D, dtype, max_B, max_L, training=training):
        took = before - torch.cuda.mem_get_info()[0]
    want = stated(D, dtype, max_B, max_L, training)
    assert want - 4 * MB <= took <= want + 4 * MB
    assert torch.cuda.mem_get_info()[0] >= before
