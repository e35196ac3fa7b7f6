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

// Whether slot s's table row names a page of the cache for page number i.
SVG_DEV bool page_of(const svg_kv_cache& c, int s, long i, int& page) {
  const int held = c.pages[s];
  if (i < 0 || i >= held || held > c.width) return false;
  page = c.table[(size_t)s * c.width + i];
  return (u32)page < (u32)c.n_pages;
}

// Whether that page may be written: no other slot holds it.  (A slot that kv_reserve refused still has the page that it
// shares.)
SVG_DEV bool own_page_of(const svg_kv_cache& c, int s, long i, int& page) {
  return page_of(c, s, i, page) && (c.refs == nullptr || c.refs[page] <= 1);
}
