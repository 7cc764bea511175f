"""The committed traffic counters (profiles/counters.json) belong to the sources that they are reported for (CPU)."""
import os
import re

import bench
from memory_bound_decode_gemv_amd import profiling


def test_the_headline_line_reports_its_traffic():
    """bench.py reports the counters only for unchanged sources; after a change to these files they are taken again
    (`bench.py --profile-kernels` under rocprofv3, then `profiling counters`)."""
    assert bench.traffic_from_profiles("gemv_q4_0_m1_28672x8192") is not None


def test_entries_name_the_headers_of_their_kernels():
    for key, (_, _, _, sources) in profiling.KERNELS.items():
        for name in sources:
            text = open(os.path.join(profiling.CSRC, name)).read()
            for header in re.findall(r'^#include "(\w+\.h)"', text, re.M):
                if header != "dg_internal.h" and os.path.exists(os.path.join(profiling.CSRC, header)):   # kernels' code
                    assert header in sources, f"{key}: {name} includes {header}"
