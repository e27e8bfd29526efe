"""A problem's offsets and block table belong to one device (with stand-ins for tensors: no GPU)."""
import pytest
import torch


class OnDevice:
    """What Problem asks of an int32 CUDA tensor."""

    is_cuda, dtype = True, torch.int32

    def __init__(self, device, shape):
        self.device_index, self.shape = device, shape

    def get_device(self):
        return self.device_index

    def dim(self):
        return len(self.shape)

    def contiguous(self):
        return self

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("devices,fits", [((0, 0, 0), True), ((1, 1, 1), True), ((0, 1, 0), False), ((0, 0, 1), False),
                                          ((1, 0, 0), False)])
def test_offsets_and_table_on_one_device(devices, fits):
    import sparse_attention_lightning_gb300 as dsa
    q, k, table = (OnDevice(d, s) for d, s in zip(devices, ((3,), (3,), (2, 4))))

    def make():
        return dsa.Problem(q, k, q_lens=[1, 1], k_lens=[9, 30], h_idx=4, d_idx=32, h=8, d_c=64, d_rope=16, top_k=8,
                           idx_dtype="e4m3", kv_dtype="bf16", block_table=table, page_size=16, num_pages=9)

    if fits:
        P = make()
        assert P._device == devices[0]
    else:
        with pytest.raises(ValueError, match="one device"):
            make()
