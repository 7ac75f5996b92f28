"""The smoke run's products of spec_linear take the kernel forms that they are there for (no GPU needed:
the choice is a function of the sizes and the device's counts)."""
import torch

import __graft_entry__ as entry
from test_linear_forms import CLUSTERS, SMS, sv  # noqa: F401

WANT = {"few tokens": ("few", False), "one CTA a tile": ("tiles", False), "split K": ("tiles", True),
        "CTA pairs": ("pairs", False)}


def test_smoke_sizes_reach_their_forms(sv):  # noqa: F811
    assert set(entry.SMOKE_LINEAR) == set(WANT)
    for name, (rows, N, K) in entry.SMOKE_LINEAR.items():
        for held in CLUSTERS:
            kind, _, splits = sv.spec_linear_form(rows, N, K, torch.float8_e4m3fn, SMS, held)
            assert (kind, splits > 1) == WANT[name], (name, kind, splits)
