"""Sizes past which the eviction's and the compaction's 32-bit row numbers would not hold are refused
before any launch (no GPU)."""
import pytest
import torch

from test_evict_host import COMPACT, EVICT, S, _accepted, _compact_args, _evict_args, base, lib  # noqa: F401

MOST = 1 << 30  # rows of a list, positions of a table


def _far(a, name, base):  # noqa: F811
    """Room for any list behind the other buffers; it is never read."""
    a[name] = base + (1 << 40)
    return a


@pytest.mark.parametrize("change", [
    {"K": MOST + 1}, {"K": (1 << 31) - 1}, {"max_pages": MOST // 1024 + 1, "page_size": 1024},
    {"max_pages": MOST // 16 + 1}, {"max_pages": (1 << 27) - 1},
])
def test_evict_refuses_more_rows_than_it_can_number(lib, base, change):  # noqa: F811
    a = _far(_evict_args(base), "kept", base)
    a.update(B=1, freed=None, n_freed=None, block_table=base + (1 << 41))
    a.update(change)
    assert lib.mla_paged_evict(*[a[n] for n in EVICT]) == S.ERR_SHAPE


def test_evict_takes_as_many_as_it_can(lib, base):  # noqa: F811
    if torch.cuda.is_available():
        return
    a = _far(_evict_args(base), "kept", base)
    a.update(B=1, freed=None, n_freed=None, block_table=base + (1 << 41), K=MOST,
             max_pages=MOST // 16)
    assert _accepted(lib.mla_paged_evict(*[a[n] for n in EVICT]))


@pytest.mark.parametrize("change", [
    {"K": MOST + 1}, {"K": (1 << 31) - 1}, {"max_pages": MOST // 1024 + 1, "page_size": 1024},
    {"max_pages": (1 << 27) - 1},
])
def test_compact_refuses_more_rows_than_it_can_number(lib, base, change):  # noqa: F811
    a = _compact_args(base)
    a.update(B=1, workspace_bytes=1 << 40)
    a.update(change)
    assert lib.mla_latent_compact(*[a[n] for n in COMPACT]) == S.ERR_SHAPE


def test_compact_takes_as_many_as_it_can(lib, base):  # noqa: F811
    if torch.cuda.is_available():
        return
    a = _compact_args(base)
    a.update(B=1, workspace_bytes=1 << 40, K=MOST, max_pages=MOST // 16)
    assert _accepted(lib.mla_latent_compact(*[a[n] for n in COMPACT]))
