"""Plain fp64 CPU oracle for Hessian-aware int4 weight quantization (GPTQ), the Bf16TrilDiagF32
Hessian codec, the e4m3 layers with block scales and the expert layout of tokens.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path (``libhq.so`` and its Python
binding) imports, links or calls this package.  Only ``tests/``, ``__graft_entry__.smoke()``
and the CPU-baseline / reference legs of ``bench.py`` may use it.

Every function is a direct, unblocked restatement of what the source pages define; see
``oracle/hq_oracle.py`` for the citations and for the readings taken where the pages are
silent.  The pages do not treat ``oracle/fp8_experts.py``'s subjects: its functions are written
from the formulas it states.  The package shares no code, header, table or constant with the
CUDA path.
"""

from .fp8_experts import *  # noqa: F401,F403
from .fp8_experts import __all__ as _fp8_experts_all
from .hq_oracle import *  # noqa: F401,F403
from .hq_oracle import __all__ as _hq_oracle_all

__all__ = [*_hq_oracle_all, *_fp8_experts_all]
