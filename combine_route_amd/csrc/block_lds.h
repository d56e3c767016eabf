// Loads from memory straight to LDS for the kernels that feed the matrix units
// from LDS: as moe_lds.h's, of 4 bytes.
#pragma once

#include "block_device.h"
#include "moe_lds.h"

namespace block {
namespace dev {

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 4 bytes a lane: lane i's to dst + 4 * i.
__device__ __forceinline__ void load4_to_lds(u32x4 rsrc, uint32_t dst, uint32_t off)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 ::"s"(dst), "v"(off), "s"(rsrc)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

}  // namespace dev
}  // namespace block
