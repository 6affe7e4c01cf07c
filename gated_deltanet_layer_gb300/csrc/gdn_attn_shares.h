// Shares of the paged attention's work and the joins of tasks that several CTAs share: plain arithmetic,
// so that a host program can walk it over any list of tasks.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

// The CTAs' shares of the units.
struct Shares {
  long long each, more, units;  // the first `more` CTAs have one unit more
  int ctas;
  GDN_HD Shares(long long units, int ctas) : units(units), ctas(ctas) {
    each = units / ctas;
    more = units - each * ctas;
  }
  GDN_HD long long first(int c) const { return c * each + (c < more ? c : more); }
  GDN_HD int owner(long long u) const {
    const long long wide = more * (each + 1);
    return u < wide ? (int)(u / (each + 1)) : (int)(more + (u - wide) / each);
  }
};

// The join of a task's parts, one for each of the CTAs c0 .. c0 + parts - 1. Up to 16 are joined at once, more in two
// levels: who finishes last of a group of about sqrt(parts) joins the group's into its first part, and
// the last of those all groups'. No CTA has many to read.
struct Join {
  int c0, parts, size, groups;
  GDN_HD Join(int c0, int c1) : c0(c0), parts(c1 - c0 + 1) {
    size = parts <= 16 ? parts : (int)ceilf(sqrtf((float)parts));
    groups = (parts + size - 1) / size;
  }
  GDN_HD int first_level() const { return groups > 1 ? 0 : 1; }
  GDN_HD int group(int cta) const { return (cta - c0) / size; }
  // What is joined at a level: `count` parts, the first part `begin` and those every `step` after it.
  GDN_HD int begin(int level, int group) const { return level == 0 ? group * size : 0; }
  GDN_HD int step(int level) const { return level == 0 || groups == 1 ? 1 : size; }
  GDN_HD int count(int level, int group) const {
    if (level == 1) return groups == 1 ? parts : groups;
    const int left = parts - group * size;
    return left < size ? left : size;
  }
  // The word of [2 ctas] in which a level's parts are counted. The next task may begin in this one's last CTA, and both be
  // joined at once: groups are numbered from c0 on, fewer than there are parts, so that none has c1's word.
  GDN_HD int word(int level, int group, int ctas) const { return level == 0 ? ctas + c0 + group : c0; }
};

}  // namespace gdn
