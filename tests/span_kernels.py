"""Which of the span kernels a call launches, from the profiler's record of it."""
import re

import torch


def kernels_of(fn):
    """fn() and the set of the span kernels that ran in it ("span_tc<128, paged>", "span_f32<64, 16 rows>"), None
    where the profiler records no kernel at all."""
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA], acc_events=True) as prof:
        result = fn()
        torch.cuda.synchronize()
    names, events = set(), prof.events()
    for e in events:
        m = re.search(r"(span_tc|span_few)_kernel<(\d+), (\w+)>|(span_f32)_kernel<(\d+), (\d+)>", e.name)
        if m and m.group(1):
            names.add(f"{m.group(1)}<{m.group(2)}, {'paged' if m.group(3) in ('true', '1') else 'dense'}>")
        elif m:
            names.add(f"{m.group(4)}<{m.group(5)}, {m.group(6)} rows>")
    return result, names if len(events) else None
