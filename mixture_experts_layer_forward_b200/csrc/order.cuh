// order.cuh -- programmatic launch order of the dense product's and dropout's kernels (ops_api.cu
// launches them with that attribute): a launch's blocks may be set up as soon as every block of the launch in front of
// it on the stream has started, and wait for that launch's end and its writes before they touch
// memory. Every thread of these kernels calls both at its start, so no launch ends before the ones
// in front of it have. Hides part of the gap between short launches (dropout of 8192 x 4096 bf16, calls
// back to back: 34.9 to 32.8 us). Not for routing: its launches fill the SMs once, and the blocks set
// up early took turns from the running ones (14.4 to 15.7 us for 16384 tokens).
#pragma once

namespace moe {

__device__ __forceinline__ void order_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void order_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

} // namespace moe
