// The paged cache on the device: its layout (svgemm_layer.h) and 16-bit types.
#pragma once
#include "../../include/svgemm_layer.h"
#include "svg_device.h"

// Elements before token t, value d of one head of a page.
SVG_DEV u32 kv_key_at(u32 t, u32 d, u32 dim) {
  return ((t >> 4) * (dim >> 5) + (d >> 5)) * 512u + (16u * ((d & 31u) >> 3) + (t & 15u)) * 8u + (d & 7u);
}
SVG_DEV u32 kv_value_at(u32 t, u32 d, u32 dim) {
  return ((t >> 5) * (dim >> 4) + (d >> 4)) * 512u + (16u * ((t & 15u) >> 2) + (d & 15u)) * 8u +
         4u * ((t & 31u) >> 4) + (t & 3u);
}

// fp32 to the cache's type, to nearest even (one rounding).
template <bool BF>
SVG_DEV u32 kv_round(float f) {
  if constexpr (BF) return (u32)__builtin_bit_cast(uint16_t, (__bf16)f);
  else return (u32)__builtin_bit_cast(uint16_t, (_Float16)f);
}
