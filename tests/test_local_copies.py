"""The library's copies into shared memory go to one block each.

Pools are any device memory that the caller has, mapped from another GPU too, and a copy that one block issues for several
is only safe on a GPU's own; so no kernel may hold such a copy, whatever launches it."""

import os
import re

from paged_decode_attention_gb300 import _build

BULK = re.compile(r"cp\.async\.bulk[^;]*")


def test_no_bulk_copy_goes_to_several_blocks():
    seen = 0
    for path in _build._sources():
        if os.path.dirname(path) != _build.CSRC:
            continue
        with open(path) as f:
            for copy in BULK.findall(f.read()):
                seen += 1
                assert "multicast" not in copy, "%s: %s" % (os.path.basename(path), copy[:120])
    assert seen > 0
