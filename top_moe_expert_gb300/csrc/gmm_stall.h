// gmm_stall.h -- failure detection in the ragged and 4-bit products, for its test.
//
// In the debug build (MOE_DEBUG_BOUNDS) moe_debug_products_stall(1) makes the
// launches that follow wait, before every tile that is not its pair's first, for a
// barrier that nothing arrives on.  The wait runs out after its limit like any
// other; the kernel reports it and ends, with the context usable.  Process-wide.
// In the release build there is no such wait.
#pragma once

#ifdef MOE_DEBUG_BOUNDS
#include <atomic>

namespace moe {
extern std::atomic<int> g_products_stall;
}

#define MOE_STALL_ARG int stall;
#define MOE_STALL_VALUE , ::moe::g_products_stall.load(std::memory_order_relaxed)
#define MOE_STALL_BARRIER uint64_t never;
#define MOE_STALL_INIT(s) tc::mbar_init(tc::smem_u32(&(s).never), 1)
#define MOE_STALL(a, s, cond)                                                                                          \
    if ((a).stall && (cond) && !tc::mbar_wait(tc::smem_u32(&(s).never), 0, &(s).abort, kWaitNs))                        \
    break
#else
#define MOE_STALL_ARG
#define MOE_STALL_VALUE
#define MOE_STALL_BARRIER
#define MOE_STALL_INIT(s)
#define MOE_STALL(a, s, cond)
#endif
