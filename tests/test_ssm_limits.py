"""Host-side checks of the state space entry points at the ends of the sizes
that include/gdn_ssm.h supports.  No GPU: only the workspace query runs."""
import itertools
import json
import os
import subprocess
import sys

from gated_deltanet_linear_pre_amd import ssm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# heads, head_dim, state_dim, n_seq, total_T, max_T
CORNERS = [(H, P, N, n, T, m) for H, P, N, n, T, share in itertools.product(
    (1, 4096), (16, 64, 128, 256), (32, 256), (1, 1 << 20), (1 << 20, (1 << 25) + 1, 1 << 26, (1 << 27) - 1, 1 << 27), (1, 3, 4096))
    for m in [T // share]]

QUERY = """
import json, sys
from gated_deltanet_linear_pre_amd import ssm
print(json.dumps([ssm.gdn_ssm_scan_workspace_bytes(ssm.make_ssm_shape(H, P, 1, N, n, T, m)) for H, P, N, n, T, m in json.load(sys.stdin)]))
"""


def test_scan_workspace_of_the_largest_sizes():
    # in a process of its own: a division by zero there would end this one
    r = subprocess.run([sys.executable, "-c", QUERY], input=json.dumps(CORNERS), capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, f"the query ended its process: {r.returncode}\n{r.stderr[-500:]}"
    for (H, P, N, n, T, m), got in zip(CORNERS, json.loads(r.stdout)):
        if T * H * -(-P // 64) >= 512 * m and m > 256:  # a 512th of the work holds the longest sequence: nothing is cut
            assert got == 0, (H, P, N, n, T, m, got)
        elif m > 256:
            state = 4 * H * (P * N + 1)  # of one segment, and its decay
            assert 2 * state <= got <= (T // 64 + n) * state + 512, (H, P, N, n, T, m, got)


def test_scan_workspace_is_asked_for():
    s = ssm.make_ssm_shape(64, 64, 8, 128, 1, 16384, 16384)
    need = ssm.gdn_ssm_scan_workspace_bytes(s)
    assert need > 0
    P = 0x10000  # an address that is never used: the call is refused
    args = [P] * 9
    assert ssm.gdn_ssm_scan(s, *args, P, workspace_bytes=need - 1, stream=0, check=False) == -4
    assert ssm.gdn_ssm_scan(s, *args, None, workspace_bytes=need, stream=0, check=False) == -1
    assert ssm.gdn_ssm_scan(s, *args, P + 128, workspace_bytes=need, stream=0, check=False) == -3
