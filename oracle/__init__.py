"""CPU oracle for multi-scale retention (test infrastructure only; see
retention_oracle.py).  Only tests/, __graft_entry__.smoke() and bench.py's
CPU legs may import it."""
from .retention_oracle import (  # noqa: F401
    backward, chunkwise, decay_mask, gated, group_norm, parallel, recurrent, rel_frobenius, rotate,
    step, swish,
)
from .block_oracle import (  # noqa: F401
    add_norm, add_norm_backward, entering, norm_gate, norm_gate_backward, norm_rows,
    norm_rows_backward, scan, scan_backward, scan_gates,
)
