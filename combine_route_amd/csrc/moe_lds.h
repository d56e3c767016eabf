// Loads from memory straight to LDS, and the waits between them and the reads,
// for the kernels that feed the matrix units from LDS.
#pragma once

#include "moe_device.h"

namespace moe {
namespace dev {

using ep::dev::u32x4;

// The end of a phase: this wave's LDS reads have returned and at most N of its
// loads are in flight; then the same holds for every wave.
template <int N>
__device__ __forceinline__ void phase_end()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ void phase_end()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// 16 bytes a lane straight to LDS: lane i's to dst + 16 * i. NT: stream. In
// assembly because the compiler makes every LDS read after the builtin wait
// for all loads in flight (it cannot tell which slice a read is of); written
// so, the only waits are the kernel's own. No register is written, so nothing
// the load does later can meet the compiler's registers, and its own counted
// waits only get stricter by loads it does not know of.
// dst is an LDS address. M0 holds it, and is named as overwritten: the
// compiler keeps no value of its own there across the statement (it warns that
// it would not hand the register out either). What is checked against the resource's
// bytes is off + soff, whichever part of it is past them (measured on gfx950,
// soff past them too).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <bool NT>
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t dst, uint32_t off, uint32_t soff)
{
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                     ::"s"(dst), "v"(off), "s"(rsrc), "s"(soff)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     ::"s"(dst), "v"(off), "s"(rsrc), "s"(soff)
                     : "memory", "m0");
}
#pragma clang diagnostic pop

// A base that every lane holds alike, and a resource over `bytes` of it, as four
// words in scalar registers: a resource the compiler takes for a lane's own
// costs a loop over the lanes at every use.
__device__ __forceinline__ u32x4 rsrc_words(const void* base, int bytes)
{
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return u32x4{(uint32_t)ep::dev::uniform((int)(uint32_t)p),
                 (uint32_t)ep::dev::uniform((int)(uint32_t)(p >> 32)) & 0xFFFFu,
                 (uint32_t)ep::dev::uniform(bytes), (uint32_t)ep::dev::kRsrcWord3};
}

}  // namespace dev
}  // namespace moe
