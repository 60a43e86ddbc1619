"""PagedCache keeps the tensors it was given: their addresses were taken when it was made."""

import pytest
import torch


def test_attributes_do_not_change_their_tensors():
    import speculative_sampling_verification_amd as sv
    k, i = torch.zeros((1, 6, 4, 2, 64)), torch.zeros(3, dtype=torch.int32)
    c = sv.PagedCache(k, k.clone(), torch.zeros((3, 5), dtype=torch.int32), i, seq_pages=i.clone(),
                      refcount=torch.zeros(6, dtype=torch.int32))
    for name in ("k", "v", "page_table", "seq_lens", "seq_pages", "refcount"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name).clone())
    with pytest.raises(AttributeError):
        c.page_size = 8
    c.steps = 1              # a caller's own note
    c.steps = 2
    c.seq_lens += 2          # in place: the same tensor
    c.seq_lens[1] = 7
    assert c.seq_lens is i and i.tolist() == [2, 7, 2]
