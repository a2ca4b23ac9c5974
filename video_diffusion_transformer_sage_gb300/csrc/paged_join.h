// paged_join.h -- which ticket counter and which workspace slot belongs to what when the few-row kernel joins the
// parts of units whose key tiles lie in several CTAs.  Plain integer arithmetic, the same on host and device.
//
// A unit's parts lie in consecutive rows of CTAs (a row: the `lock` CTAs that take K/V heads side by side), one
// part to a row.  Each part is left in a slot; the CTA that draws the last ticket of a group of parts joins them.  Up to
// kJoinAtOnce parts are one group; more are dealt evenly to about sqrt(parts) groups, whose results are joined by the CTA
// that draws the last of the groups' tickets.
//
// What belongs to one unit alone: a row holds at most two parts, the end of one unit and the beginning of a
// later one, and whatever begins there is that later unit's.  A group's counter and slot are those of its first part's row.
// So no group but a unit's first may begin in the unit's last row, where the next unit may begin: with at
// least two parts to every group none does.
#pragma once

#ifdef __CUDACC__
#define SAGE_HD __host__ __device__ __forceinline__
#else
#define SAGE_HD inline
#endif

namespace sage {

// The most CTAs whose partial results the workspace holds, and its slots.
constexpr int kPagedMaxCtas = 320;
constexpr int kPagedSlots = 2 * kPagedMaxCtas;
// Parts take two slots per CTA from the front, joined groups one from the back.
constexpr int kFewMaxCtas = (kPagedSlots - 1) / 3;
constexpr int kJoinAtOnce = 16;

SAGE_HD int join_groups(int parts) {
  if (parts <= kJoinAtOnce) return 1;
  int per = 5;
  while (per * per < parts) ++per;
  return (parts + per - 1) / per;
}
// Group g's first part (of group `groups`: the number of parts).  Sizes differ by one at most, so above 16 parts, with at
// most per groups of about per >= 5 parts, none has fewer than three.
SAGE_HD int join_first(int parts, int groups, int g) { return parts * g / groups; }
// The group of a part: the largest g with join_first(g) <= part.
SAGE_HD int join_group_of(int parts, int groups, int part) { return ((part + 1) * groups - 1) / parts; }
// The tickets of a group whose first part lies in CTA row `row`, and those of the groups of a unit that begins in `row`.
SAGE_HD int join_counter(int row, int lock, int col) { return row * lock + col; }
SAGE_HD int join_unit_counter(int row, int lock, int col) { return kPagedMaxCtas + row * lock + col; }
// The slot of a part in CTA row `row` (`head`: the part that begins its unit), and that of a joined group.
SAGE_HD int join_part_slot(int row, int lock, int col, bool head) { return (row * lock + col) * 2 + (head ? 1 : 0); }
SAGE_HD int join_group_slot(int row, int lock, int col) { return kPagedSlots - 1 - (row * lock + col); }

}  // namespace sage
